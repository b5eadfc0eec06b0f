// Calls of the dense operators that the library must refuse before any launch, and the
// host-only ones over a grid of shapes; built with the host sanitizers and run without a GPU.
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
  for (int32_t n : {1, 15, 16, 129, 18944, 1 << 20, 1 << 24})
    for (int32_t k : {1, 16, 127, 128, 129, 5120, 18944, 1 << 24})
      for (int32_t gated : {0, 1}) {
        mbq_fp8_desc d;
        if (mbq_fp8_describe(n, k, gated, &d) != MBQ_OK) continue;
        EXPECT(d.total_bytes > uint64_t(n) * uint64_t(k));
        for (int32_t t : {0, 1, 4, 16, 17, 64, 65, 333, 4096, 1 << 21})
          for (mbq_dtype x : {MBQ_F32, MBQ_BF16, MBQ_E4M3}) {
            size_t b = 0;
            EXPECT(mbq_fp8_linear_workspace(&d, t, x, &b) == MBQ_OK);
            EXPECT(t > 0 || b == 0);
          }
      }
  mbq_fp8_desc d, g;
  EXPECT(mbq_fp8_describe(100, 304, 0, &d) == MBQ_OK && mbq_fp8_describe(100, 304, 1, &g) == MBQ_OK);
  EXPECT(mbq_fp8_describe(0, 8, 0, &d) == MBQ_ERR_SHAPE && mbq_fp8_describe(8, 8, 3, &d) == MBQ_ERR_ARG);
  EXPECT(mbq_fp8_describe(100, 304, 0, nullptr) == MBQ_ERR_ARG);
  EXPECT(mbq_fp8_pack(&d, 1, fake(0), MBQ_F32, nullptr, fake(0), nullptr, nullptr) == MBQ_ERR_ARG);
  EXPECT(mbq_fp8_pack(&g, 2, fake(0), MBQ_F32, nullptr, fake(0), nullptr, nullptr) == MBQ_ERR_ARG);
  EXPECT(mbq_fp8_pack(nullptr, 0, fake(0), MBQ_F32, nullptr, fake(0), nullptr, nullptr) == MBQ_ERR_ARG);
  EXPECT(mbq_fp8_quantize(4, 8, fake(0), mbq_dtype(9), 8, fake(0), 8, ffake(0), nullptr) == MBQ_ERR_ARG);
  EXPECT(mbq_fp8_quantize(4, 8, fake(0), MBQ_F32, 7, fake(0), 8, ffake(0), nullptr) == MBQ_ERR_SHAPE);
  EXPECT(mbq_fp8_linear(&g, fake(0), 4, fake(0), MBQ_BF16, 304, nullptr, fake(0), MBQ_BF16, fake(0), 1 << 30, nullptr) ==
         MBQ_ERR_UNSUPPORTED);
  EXPECT(mbq_fp8_linear(&d, fake(0), 4, fake(0), MBQ_E4M3, 304, nullptr, fake(0), MBQ_BF16, nullptr, 0, nullptr) == MBQ_ERR_ARG);
  EXPECT(mbq_fp8_linear(&d, fake(0), 4, fake(8), MBQ_E4M3, 304, ffake(0), fake(0), MBQ_BF16, nullptr, 0, nullptr) == MBQ_ERR_ARG);
  EXPECT(mbq_fp8_linear(&d, fake(0), 64, fake(0), MBQ_BF16, 304, nullptr, fake(0), MBQ_BF16, nullptr, 0, nullptr) ==
         MBQ_ERR_WORKSPACE);
  EXPECT(mbq_fp8_gated(&g, fake(0), 4, fake(0), MBQ_BF16, 304, nullptr, mbq_act(7), fake(0), MBQ_BF16, nullptr, 0, nullptr) ==
         MBQ_ERR_ARG);
  mbq_block_norm_args a = {};
  a.t = 4;
  a.k = 100;
  a.x = fake(0);
  a.h = fake(0);
  a.ldx = a.ldr = a.ldy = a.ldh = 100;
  a.eps = 0.f;
  EXPECT(mbq_block_norm(&a, nullptr) == MBQ_ERR_RANGE);
  a.eps = NAN;
  EXPECT(mbq_block_norm(&a, nullptr) == MBQ_ERR_RANGE);
  a.eps = 1e-6f;
  a.ldx = 99;
  EXPECT(mbq_block_norm(&a, nullptr) == MBQ_ERR_SHAPE);
  a.ldx = 100;
  a.gate_kind = 9;
  EXPECT(mbq_block_norm(&a, nullptr) == MBQ_ERR_ARG);
  EXPECT(mbq_block_norm(nullptr, nullptr) == MBQ_ERR_ARG);
  for (int32_t t : {0, 1, 3, 64, 1030, 1 << 21})
    for (int32_t v : {1, 7, 2048, 131072, 1 << 28})
      for (int32_t top : {0, 1, 64}) {
        size_t b = 0;
        EXPECT(mbq_token_logprobs_workspace(t, v, top, &b) == (top > v ? MBQ_ERR_SHAPE : MBQ_OK));
      }
  EXPECT(mbq_token_logprobs(2, 500, fake(0), MBQ_BF16, 499, fake(0), 64, 1.f, 0, ffake(0), ffake(0), ifake(0), nullptr, nullptr,
                            nullptr, 0, nullptr) == MBQ_ERR_SHAPE);
  EXPECT(mbq_token_logprobs(2, 500, fake(0), MBQ_BF16, 500, fake(0), 16, 1.f, 0, ffake(0), ffake(0), ifake(0), nullptr, nullptr,
                            nullptr, 0, nullptr) == MBQ_ERR_ARG);
  EXPECT(mbq_token_logprobs(2, 500, fake(0), MBQ_BF16, 500, fake(0), 64, -1.f, 0, ffake(0), ffake(0), ifake(0), nullptr, nullptr,
                            nullptr, 0, nullptr) == MBQ_ERR_RANGE);
  EXPECT(mbq_token_logprobs(1, 1 << 19, fake(0), MBQ_F32, 1 << 19, fake(0), 64, 1.f, 0, ffake(0), ffake(0), ifake(0), nullptr,
                            nullptr, nullptr, 0, nullptr) == MBQ_ERR_WORKSPACE);
  std::printf(failed ? "failed\n" : "ok\n");
  return failed;
}
