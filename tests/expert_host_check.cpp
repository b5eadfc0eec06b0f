// Calls of the 8-bit integer linear and the expert operators that the library must refuse before
// any launch, and the host-only ones over a grid of shapes; built with the host sanitizers and
// run without a GPU.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "mbq.h"

static int failed = 0;
#define EXPECT(c)                                               \
  do {                                                          \
    if (!(c)) {                                                 \
      std::printf("line %d: %s\n", __LINE__, #c);               \
      failed = 1;                                               \
    }                                                           \
  } while (0)

static void* fake(uintptr_t off) { return reinterpret_cast<void*>(uintptr_t(0x7F0000000000) + off); }
static float* ffake(uintptr_t off) { return static_cast<float*>(fake(off)); }
static int32_t* ifake(uintptr_t off) { return static_cast<int32_t*>(fake(off)); }

int main() {
  for (int32_t n : {-1, 0, 1, 15, 17, 1000, 18944, 1 << 20, 1 << 24, INT32_MAX})
    for (int32_t k : {0, 1, 16, 127, 129, 5120, (1 << 17) - 1, 1 << 17, INT32_MAX})
      for (int32_t gated : {0, 1})
        for (int32_t experts : {0, 1, 2, 40, 128, 1024, 1025}) {
          mbq_int8_desc d;
          if (mbq_int8_describe(n, k, gated, experts, &d) != MBQ_OK) continue;
          EXPECT(d.total_bytes > uint64_t(n) * uint64_t(k) * (gated + 1) * experts && d.scales_offset == d.expert_stride * experts);
          for (int32_t t : {0, 1, 2, 9, 17, 64, 333, 4096, 1 << 21})
            for (int32_t p : {0, 1, 16, 17, 4096, 1 << 24})
              for (mbq_dtype x : {MBQ_F32, MBQ_BF16, MBQ_INT8})
                for (int32_t grouped : {0, 1}) {
                  if (!grouped && (experts != 1 || p != t)) continue;
                  size_t b = 1;
                  EXPECT(mbq_int8_workspace(&d, t, p, grouped, x, &b) == MBQ_OK);
                  EXPECT(p > 0 || b == 0);
                }
        }
  mbq_int8_desc d, g, e;
  EXPECT(mbq_int8_describe(100, 304, 0, 1, &d) == MBQ_OK && mbq_int8_describe(100, 304, 1, 1, &g) == MBQ_OK);
  EXPECT(mbq_int8_describe(100, 304, 0, 5, &e) == MBQ_OK && mbq_int8_describe(100, 304, 0, 5, nullptr) == MBQ_ERR_ARG);
  EXPECT(mbq_int8_describe(100, 304, 2, 5, &d) == MBQ_ERR_ARG && mbq_int8_describe(100, 1 << 17, 0, 1, &d) != MBQ_OK);
  EXPECT(mbq_int8_describe(100, 304, 0, 1, &d) == MBQ_OK);
  EXPECT(mbq_int8_pack(&d, 1, fake(0), MBQ_F32, nullptr, fake(0), nullptr, nullptr) == MBQ_ERR_ARG);
  EXPECT(mbq_int8_pack(&g, 2, fake(0), MBQ_F32, nullptr, fake(0), nullptr, nullptr) == MBQ_ERR_ARG);
  EXPECT(mbq_int8_pack(&d, 0, fake(0), MBQ_INT8, nullptr, fake(0), nullptr, nullptr) == MBQ_ERR_ARG);
  EXPECT(mbq_int8_pack(nullptr, 0, fake(0), MBQ_F32, nullptr, fake(0), nullptr, nullptr) == MBQ_ERR_ARG);
  EXPECT(mbq_int8_quantize(4, 8, fake(0), mbq_dtype(9), 8, fake(0), 8, ffake(0), nullptr) == MBQ_ERR_ARG);
  EXPECT(mbq_int8_quantize(4, 8, fake(0), MBQ_F32, 7, fake(0), 8, ffake(0), nullptr) == MBQ_ERR_SHAPE);
  size_t b = 0;
  EXPECT(mbq_int8_workspace(&e, 4, 4, 0, MBQ_F32, &b) != MBQ_OK && mbq_int8_workspace(&d, 4, 5, 0, MBQ_F32, &b) != MBQ_OK);
  EXPECT(mbq_int8_workspace(&d, 4, 4, 0, MBQ_F32, nullptr) == MBQ_ERR_ARG);

  EXPECT(mbq_int8_linear(&d, fake(0), nullptr, nullptr) == MBQ_ERR_ARG);
  const auto with = [&](auto set) {
    mbq_int8_args a = {};
    a.t = a.p = 40;
    a.x_dtype = MBQ_INT8;
    a.y_dtype = MBQ_BF16;
    a.x = fake(0);
    a.x_scale = ffake(0);
    a.y = fake(0);
    a.ldx = 304;
    a.workspace = fake(0);
    a.ws_bytes = 1 << 30;
    const mbq_int8_desc* desc = &d;
    set(a, desc);
    return mbq_int8_linear(desc, fake(0), &a, nullptr);
  };
  EXPECT(with([](auto& a, auto&) { a.x_scale = nullptr; }) == MBQ_ERR_ARG);
  EXPECT(with([](auto& a, auto&) { a.x = nullptr; }) == MBQ_ERR_ARG);
  EXPECT(with([](auto& a, auto&) { a.x = fake(8); }) == MBQ_ERR_ARG);
  EXPECT(with([](auto& a, auto&) { a.y = nullptr; }) == MBQ_ERR_ARG);
  EXPECT(with([](auto& a, auto&) { a.y_dtype = MBQ_E4M3; }) == MBQ_ERR_ARG);
  EXPECT(with([](auto& a, auto&) { a.reserved = 1; }) == MBQ_ERR_ARG);
  EXPECT(with([](auto& a, auto&) { a.ldx = 303; }) == MBQ_ERR_SHAPE);
  EXPECT(with([](auto& a, auto&) { a.p = 41; }) != MBQ_OK);
  EXPECT(with([](auto& a, auto&) { a.t = a.p = -1; }) != MBQ_OK);
  EXPECT(with([](auto& a, auto&) { a.rows = ifake(0); }) != MBQ_OK);
  EXPECT(with([](auto& a, auto&) { a.act = 7; }) != MBQ_OK);
  EXPECT(with([&](auto&, auto& desc) { desc = &e; }) != MBQ_OK);
  EXPECT(with([](auto& a, auto&) { a.x_dtype = MBQ_BF16; a.x_scale = nullptr; a.ws_bytes = 16; }) == MBQ_ERR_WORKSPACE);
  EXPECT(with([](auto& a, auto&) { a.x_dtype = MBQ_BF16; a.x_scale = nullptr; a.workspace = nullptr; }) == MBQ_ERR_WORKSPACE);

  for (int32_t t : {0, 1, 64, 65, 4096, 4097, 1 << 21})
    for (int32_t experts : {1, 7, 64, 65, 1024}) EXPECT(mbq_expert_route_workspace(t, experts, &b) == MBQ_OK);
  EXPECT(mbq_expert_route_workspace(4, 1025, &b) != MBQ_OK && mbq_expert_route_workspace(-1, 8, &b) != MBQ_OK);
  EXPECT(mbq_expert_route_workspace(4, 8, nullptr) == MBQ_ERR_ARG);
  const auto route = [&](int32_t t, int32_t experts, mbq_dtype dtype, int64_t ld, int32_t top, int32_t score, float scale, size_t ws) {
    return mbq_expert_route(t, experts, fake(0), dtype, ld, top, mbq_score(score), 1, scale, ifake(0), ffake(0), ifake(0), ifake(0),
                            ifake(0), fake(0), ws, nullptr);
  };
  EXPECT(route(100, 8, MBQ_INT8, 8, 2, 0, 1.f, 1 << 20) == MBQ_ERR_ARG && route(100, 8, MBQ_F32, 8, 2, 5, 1.f, 1 << 20) == MBQ_ERR_ARG);
  EXPECT(route(100, 8, MBQ_F32, 7, 2, 0, 1.f, 1 << 20) == MBQ_ERR_SHAPE && route(100, 8, MBQ_F32, 8, 9, 0, 1.f, 1 << 20) == MBQ_ERR_SHAPE);
  EXPECT(route(100, 8, MBQ_F32, 8, 0, 0, 1.f, 1 << 20) == MBQ_ERR_SHAPE && route(100, 1025, MBQ_F32, 1025, 2, 0, 1.f, 1 << 20) != MBQ_OK);
  EXPECT(route(100, 64, MBQ_F32, 64, 33, 0, 1.f, 1 << 20) != MBQ_OK && route(100, 8, MBQ_F32, 8, 2, 0, NAN, 1 << 20) != MBQ_OK);
  EXPECT(route(4096, 128, MBQ_F32, 128, 8, 0, 1.f, 16) == MBQ_ERR_WORKSPACE);
  const auto combine = [&](int32_t n, int32_t top, int32_t p, int64_t ldr, int64_t ldy, void* y) {
    return mbq_expert_combine(5, n, top, p, fake(0), MBQ_BF16, ldr, ffake(0), ifake(0), nullptr, MBQ_BF16, 0, y, ldy, nullptr);
  };
  EXPECT(combine(100, 2, 10, 99, 100, fake(0)) == MBQ_ERR_SHAPE && combine(100, 2, 10, 100, 99, fake(0)) == MBQ_ERR_SHAPE);
  EXPECT(combine(100, 33, 10, 100, 100, fake(0)) != MBQ_OK && combine(100, 0, 10, 100, 100, fake(0)) != MBQ_OK);
  EXPECT(combine(0, 2, 10, 100, 100, fake(0)) != MBQ_OK && combine(100, 2, -1, 100, 100, fake(0)) != MBQ_OK);
  EXPECT(combine(100, 2, 10, 100, 100, nullptr) == MBQ_ERR_ARG);
  std::printf(failed ? "failed\n" : "ok\n");
  return failed;
}
