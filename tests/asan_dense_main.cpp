// Drives the dense FFN block's host code with valid and invalid arguments, where no GPU is visible: a valid call then ends in
// NM_ERR_HIP at its first launch, and no device address is read.  Built with AddressSanitizer by tests/test_dense_host_asan.py.
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <memory>
#include <vector>

#include "nmsparse.h"

static int failures = 0;
#define EXPECT(call, want)                                                                  \
  do {                                                                                      \
    const int got_ = (int)(call);                                                           \
    if (got_ != (int)(want)) {                                                              \
      std::printf("%s:%d: %s gave %d, not %d\n", __FILE__, __LINE__, #call, got_, (int)(want)); \
      ++failures;                                                                           \
    }                                                                                       \
  } while (0)

static char* const P = (char*)0x100000000;   // device addresses, never read here

// n tensors of which every `hole`-th is empty, 4096 bytes apart or more; the arrays are exactly as long as the call may read
static void clip(int64_t n, int64_t count, int64_t hole, bool in_place) {
  std::unique_ptr<nm_dtype[]> dt(new nm_dtype[n]), odt(new nm_dtype[n]);
  std::unique_ptr<const void*[]> in(new const void*[n]);
  std::unique_ptr<void*[]> out(new void*[n]);
  std::unique_ptr<int64_t[]> counts(new int64_t[n]);
  char* at = P;
  for (int64_t i = 0; i < n; ++i) {
    dt[i] = i % 2 ? NM_BF16 : NM_F32;
    odt[i] = in_place ? dt[i] : NM_F32;
    counts[i] = hole && i % hole == 0 ? 0 : count;
    in[i] = counts[i] ? at : nullptr;
    at += count * 4 + 4096;
    out[i] = in_place ? const_cast<void*>(in[i]) : at;
    at += in_place ? 0 : count * 4 + 4096;
  }
  float* norm = (float*)(P - 4096);
  int64_t need = -1;
  EXPECT(grad_work_bytes(n, counts.get(), &need), NM_OK);
  if (need < 0) ++failures;
  void* work = P - (1 << 28);
  EXPECT(grad_norm(n, dt.get(), in.get(), counts.get(), norm, work, need, nullptr), NM_ERR_HIP);
  EXPECT(grad_clip(n, dt.get(), in.get(), counts.get(), 1.f, 0, norm, odt.get(), out.get(), work, need, nullptr), NM_ERR_HIP);
  const bool any = hole == 0 || (hole > 1 && n > 1);
  EXPECT(grad_clip(n, dt.get(), in.get(), counts.get(), 1.f, 1, norm, odt.get(), out.get(), nullptr, 0, nullptr), any ? NM_ERR_HIP : NM_OK);
  if (need) EXPECT(grad_norm(n, dt.get(), in.get(), counts.get(), norm, work, need - 1, nullptr), NM_ERR_SHAPE);
  EXPECT(grad_clip(n, dt.get(), in.get(), counts.get(), NAN, 0, norm, odt.get(), out.get(), work, need, nullptr), NM_ERR_UNSUPPORTED);
  if (any && n > 1) {   // the last tensor again, and a work memory or a norm inside one
    int64_t last = n - 1;
    while (last > 0 && !counts[last]) --last;
    int64_t first = 0;
    while (first < last && !counts[first]) ++first;
    if (first < last && dt[first] == dt[last]) {
      out[first] = out[last];
      EXPECT(grad_clip(n, dt.get(), in.get(), counts.get(), 1.f, 0, norm, odt.get(), out.get(), work, need, nullptr), NM_ERR_SHAPE);
    }
    EXPECT(grad_clip(n, dt.get(), in.get(), counts.get(), 1.f, 0, (float*)out[last], odt.get(), out.get(), work, need, nullptr), NM_ERR_SHAPE);
  }
}

int main() {
  for (int64_t n : {1, 2, 31, 32, 33, 159, 160, 161, 320, 321, 5000, 65536})
    for (int64_t count : {1, 5, 409, 16384, 16385, 70000})
      for (int64_t hole : {0, 1, 2, 7})
        for (bool in_place : {true, false}) clip(n, count, hole, in_place);
  clip(3, int64_t(1) << 33, 0, true);
  clip(2, int64_t(1) << 47, 0, false);   // more chunks than a table counts in 32 bits
  int64_t huge[2] = {INT64_MAX / 2, 1}, need;
  EXPECT(grad_work_bytes(2, huge, &need), NM_ERR_SHAPE);
  EXPECT(grad_work_bytes(65537, huge, &need), NM_ERR_SHAPE);

  void *A = P, *B = P + (int64_t(1) << 40), *C = P + (int64_t(2) << 40), *D = P + (int64_t(3) << 40), *W = P + (int64_t(4) << 40);
  const int64_t sizes[] = {1, 7, 16, 33, 1000, 4096, 131073, 5000000, INT32_MAX};
  for (int64_t M : sizes)
    for (int64_t N : sizes)
      for (int64_t K : sizes)
        for (int al = 0; al < 2; ++al)
          for (int c = 0; c < 3; ++c) {
            need = -1;
            EXPECT(linear_work_bytes((nm_linear)c, M, N, K, al, &need), NM_OK);
            if (need < 0) {
              std::printf("work of %d %lld %lld %lld\n", c, (long long)M, (long long)N, (long long)K);
              ++failures;
            }
          }
  for (int64_t M : {1, 16, 17, 300, 5000})
    for (int64_t N : {1, 24, 999, 4096})
      for (int64_t K : {1, 8, 777, 8192})
        for (int act = 0; act < 4; ++act)
          for (int64_t room : {int64_t(0), int64_t(1) << 40}) {
            EXPECT(linear_fwd(NM_BF16, A, K, B, K, NM_F32, D, (nm_act)act, nullptr, 0, M, N, K, NM_BF16, C, N, D, N, W, room, nullptr),
                   NM_ERR_HIP);
            EXPECT(linear_bwd_x(NM_BF16, A, N, B, K, D, K, (nm_act)act, M, N, K, NM_F32, C, K, W, room, nullptr), NM_ERR_HIP);
            EXPECT(linear_bwd_w(NM_BF16, A, N, B, K, M, N, K, 1, NM_F32, C, K, W, room, nullptr), NM_ERR_HIP);
            EXPECT(linear_bwd_act(NM_BF16, A, N, B, N, (nm_act)act, M, N, C, N, (float*)D, W, int64_t(1) << 40, nullptr), NM_ERR_HIP);
          }
  for (int64_t T : {1, 3, 513, 70000})
    for (int64_t N : {1, 512, 513, 1024, 2048, 4096, 8192, 16384}) {
      int64_t q = (N + 127) / 128 * 128;
      EXPECT(rms_norm(NM_BF16, A, N, nullptr, 0, NM_F32, B, 1e-5f, T, N, nullptr, 0, C, N, nullptr, nullptr), NM_ERR_HIP);
      EXPECT(rms_norm_fp8(NM_F32, A, N, nullptr, 0, NM_BF16, B, 1e-5f, T, N, NM_E4M3, (uint8_t*)C, q, (float*)D, T, nullptr, 0, nullptr, 0,
                          nullptr, nullptr), NM_ERR_HIP);
      EXPECT(rms_norm_bwd_work_bytes(T, N, &need), NM_OK);
      EXPECT(rms_norm_bwd(NM_BF16, A, N, B, N, NM_F32, D, (float*)D, nullptr, 0, T, N, C, N, (float*)D, W, need, nullptr), NM_ERR_HIP);
      if (need) EXPECT(rms_norm_bwd(NM_BF16, A, N, B, N, NM_F32, D, (float*)D, nullptr, 0, T, N, C, N, (float*)D, W, need - 1, nullptr), NM_ERR_SHAPE);
    }
  if (failures) return 1;
  std::printf("asan dense ok\n");
  return 0;
}
