// Host-side exercise of the mixture-of-experts calls under AddressSanitizer (built and run by
// tests/test_moe_host_asan.py where no GPU is visible): invalid arguments return their status before any
// launch; valid ones with placeholder device addresses reach the launchers, which report the missing
// device (NM_ERR_HIP).
#include <stdint.h>
#include <stdio.h>

#include "nmsparse.h"

static int failures = 0;
#define EXPECT(expr, want)                                                                   \
  do {                                                                                       \
    const int got_ = (int)(expr);                                                            \
    if (got_ != (int)(want)) {                                                               \
      fprintf(stderr, "line %d: %s returned %d, expected %d\n", __LINE__, #expr, got_, (int)(want)); \
      ++failures;                                                                            \
    }                                                                                        \
  } while (0)

int main() {
  void* P = (void*)(uintptr_t)0x10000;   // never dereferenced on the host
  uint8_t* U = (uint8_t*)P;
  float* F = (float*)P;
  int32_t* I = (int32_t*)P;
  const nm_status H = NM_ERR_HIP;
  for (int dt = 0; dt < 2; ++dt) {
    const nm_dtype d = (nm_dtype)dt;
    const int shapes[][2] = {{64, 8}, {256, 8}, {200, 30}, {1024, 64}};
    for (const auto& s : shapes) {
      EXPECT(moe_route(d, P, s[0], 5, s[0], NM_SIGMOID, F, 1, 1, 2, s[1], 1, 1.f, I, F, 0), H);
      EXPECT(moe_route_bwd(d, P, s[0], 5, s[0], NM_SOFTMAX, s[1], 0, 1.f, I, F, F, P, s[0], 0), H);
    }
    EXPECT(moe_route(d, P, 63, 5, 64, NM_SOFTMAX, 0, 1, 1, 2, 8, 1, 1.f, I, F, 0), NM_ERR_SHAPE);
    for (int fmt = 0; fmt < 2; ++fmt) {
      const nm_fp8 f = (nm_fp8)fmt;
      EXPECT(fp8_quantize(d, P, 256, 64, I, 3, P, 256, 5000, 256, f, U, 256, F, 5000, 0), H);
      EXPECT(fp8_quantize(d, P, 203, 64, 0, 1, 0, 0, 64, 203, f, U, 256, F, 64, 0), H);
      EXPECT(fp8_quantize_t(d, P, 256, 64, 0, 1, 0, 0, 64, 256, f, U, 128, F, 256, 0), H);
      EXPECT(fp8_quantize_t(d, P, 256, 64, 0, 1, 0, 0, 64, 256, f, U, 127, F, 256, 0), NM_ERR_SHAPE);
      EXPECT(fp8_quantize_weight(d, P, 256, 3, 100, 256, f, U, 256, F, U, 128, F, 0), H);
    }
    EXPECT(moe_combine(d, P, 64, 16, I, F, 4, 4, 64, P, 64, 0), H);
    EXPECT(moe_combine_bwd(d, P, 64, P, 64, 16, I, I, F, 4, 4, 64, P, 64, F, 0), H);
    for (int fa = 0; fa < 2; ++fa)
      for (int fb = 0; fb < 2; ++fb) {
        const nm_fp8 a = (nm_fp8)fa, b = (nm_fp8)fb;
        const int64_t ms[] = {1, 40, 400, 9000};
        for (int64_t m : ms) {
          EXPECT(fp8_gemm_nt(a, U, 256, F, m, b, U, 256, F, 2, 128, m, 512, 256, d, P, 512, 0), H);
          EXPECT(fp8_gemm_nt(a, U, 256, F, m, b, U, 256, F, 512, 1, m, 512, 256, d, P, 512, 0), H);
          EXPECT(fp8_gemm_nt(a, U + 1, 255, F, m, b, U, 255, F, 512, 1, m, 512, 250, d, P, 512, 0), H);
          EXPECT(fp8_gemm_nt_grouped(a, U, 256, F, m, b, U, 256, F, 2, I, 8, m, 512, 256, d, P, 512, 0), H);
        }
        EXPECT(fp8_gemm_nt_grouped_k(a, U, 1024, F, 64, b, U, 1024, F, 64, I, 8, 64, 64, 1024, d, P, 64, 0), H);
        EXPECT(fp8_gemm_nt_grouped_k(a, U, 1024, F, 64, b, U, 1024, F, 64, I, 8, 64, 64, 1000, d, P, 64, 0),
               NM_ERR_SHAPE);
      }
  }
  int64_t bytes = -1;
  EXPECT(moe_plan_work_bytes(8192, 8, 256, &bytes), NM_OK);
  EXPECT(bytes > 0, 1);
  EXPECT(moe_plan(I, 8192, 8, 256, 128, I, I, I, 8192 * 8 + 256 * 128, I, P, bytes, 0), H);
  EXPECT(moe_plan(I, 8192, 8, 256, 128, I, I, I, 8192 * 8 + 256 * 128, I, P, bytes - 1, 0), NM_ERR_SHAPE);
  EXPECT(moe_plan(I, 4, 8, 64, 1, I, I, I, 32, I, 0, 0, 0), H);
  if (failures) return 1;
  printf("asan moe ok\n");
  return 0;
}
