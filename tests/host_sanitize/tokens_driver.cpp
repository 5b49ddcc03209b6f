// Host-only exercise of the validation and planning code of the plan, append
// and chunk calls, built with AddressSanitizer and UndefinedBehaviorSanitizer
// (tests/test_host_sanitizers_tokens.py). Every call fails validation or only
// plans a workspace: no HIP call is reached.
#include <math.h>
#include <stdio.h>

#include "entmaxkv.h"

static int failures = 0;

static void expect(int got, int want, const char* what, int line) {
  if (got != want) {
    fprintf(stderr, "line %d: %s returned %d, expected %d\n", line, what, got, want);
    ++failures;
  }
}
#define EXPECT(call, want) expect((call), (want), #call, __LINE__)

int main() {
  void* d = reinterpret_cast<void*>(uintptr_t(1) << 20);
  void* e = reinterpret_cast<void*>((uintptr_t(1) << 20) + 4096);
  void* mis = reinterpret_cast<void*>((uintptr_t(1) << 20) + 8);
  const int32_t* ci = static_cast<const int32_t*>(d);
  int32_t* oi = static_cast<int32_t*>(e);
  const float* cf = static_cast<const float*>(d);
  const double* cd = static_cast<const double*>(d);
  const size_t big = size_t(1) << 60;

  // workspace plans over the supported set, up to the largest sizes
  for (int D : {64, 128})
    for (int ps : {16, 64})
      for (int G : {1, 2, 4, 8})
        for (int Hkv : {1, 8})
          for (int mp : {1, 7, 4096, 262144})
            for (int dt = 0; dt < 2; ++dt)
              for (int B : {1, 16, 300, 65536, (1 << 24) / 64})
                for (int N : {1, 63, 64, 4097, 1 << 20, (1 << 24) - 1})
                  for (float alpha : {1.0001f, 1.25f, 1.5f, 2.0f, 1e30f}) {
                    if ((long long)B * Hkv * G > (1LL << 24)) continue;
                    entmaxkv_shape s = {B, Hkv * G, Hkv, D, ps, mp, 0x7fffffff / ps, dt};
                    size_t n = 0;
                    const int rc = entmaxkv_entmax_chunk_ws(&s, N, alpha, &n);
                    if (rc != ENTMAXKV_OK && rc != ENTMAXKV_ERR_UNSUPPORTED) ++failures;
                    // a list entry and a part of every row, at least
                    if (rc == ENTMAXKV_OK && n < (size_t)N * Hkv * G * (128 * 8 + 16)) ++failures;
                  }

  entmaxkv_shape s = {4, 32, 8, 128, 32, 4096, 16384, ENTMAXKV_BF16};
  size_t n = 0;
  EXPECT(entmaxkv_entmax_chunk_ws(nullptr, 1, 1.5f, &n), ENTMAXKV_ERR_INVALID);
  EXPECT(entmaxkv_entmax_chunk_ws(&s, 1, 1.5f, nullptr), ENTMAXKV_ERR_INVALID);
  for (int bad : {0, -1, -0x7fffffff - 1}) {
    EXPECT(entmaxkv_entmax_chunk_ws(&s, bad, 1.5f, &n), ENTMAXKV_ERR_INVALID);
    EXPECT(entmaxkv_entmax_chunk(&s, d, 1, bad, ci, d, d, ci, ci, 1.5f, e, nullptr, nullptr, d, big,
                                 0, 0),
           ENTMAXKV_ERR_INVALID);
    EXPECT(entmaxkv_plan_tokens(&s, bad, ci, ci, ci, 8, ci, oi, oi, oi, oi, oi, oi, 0, 0),
           ENTMAXKV_ERR_INVALID);
  }
  EXPECT(entmaxkv_entmax_chunk(&s, d, 1, 8, ci, d, d, ci, ci, NAN, e, nullptr, nullptr, d, big, 0, 0),
         ENTMAXKV_ERR_INVALID);
  EXPECT(entmaxkv_entmax_chunk(&s, mis, 1, 8, ci, d, d, ci, ci, 1.5f, e, nullptr, nullptr, d, big, 0,
                               0),
         ENTMAXKV_ERR_INVALID);
  EXPECT(entmaxkv_entmax_chunk(&s, d, 7, 8, ci, d, d, ci, ci, 1.5f, e, nullptr, nullptr, d, big, 0, 0),
         ENTMAXKV_ERR_UNSUPPORTED);
  EXPECT(entmaxkv_entmax_chunk(&s, d, 1, 8, ci, d, d, ci, ci, 1.5f, e, nullptr, nullptr, nullptr, big,
                               0, 0),
         ENTMAXKV_ERR_WORKSPACE);
  EXPECT(entmaxkv_plan_tokens(&s, 0x7fffffff, ci, ci, ci, 8, ci, oi, oi, oi, oi, oi, oi, 0, 0),
         ENTMAXKV_ERR_UNSUPPORTED);
  EXPECT(entmaxkv_plan_tokens(&s, 8, ci, ci, ci, -1, ci, oi, oi, oi, oi, oi, oi, 0, 0),
         ENTMAXKV_ERR_INVALID);
  EXPECT(entmaxkv_plan_tokens(&s, 8, ci, ci, nullptr, 1, ci, oi, oi, oi, oi, oi, oi, 0, 0),
         ENTMAXKV_ERR_INVALID);

  const int64_t huge = INT64_MAX;
  for (int64_t stride : {int64_t(0), int64_t(-4096), INT64_MIN, huge, int64_t(4100)}) {
    entmaxkv_append a = {8, 1, 0, 128, 1, 0, stride, 6144, 6144, 1e-6f, 1.0f};
    EXPECT(entmaxkv_append_kv(&s, &a, d, d, d, ci, ci, cd, nullptr, cf, cf, e, d, d, 0, 0),
           ENTMAXKV_ERR_INVALID);
  }
  entmaxkv_append a = {8, 1, 0, 128, 1, 0, 6144, 6144, 6144, 1e-6f, 1.0f};
  EXPECT(entmaxkv_append_kv(&s, nullptr, d, d, d, ci, ci, cd, nullptr, cf, cf, e, d, d, 0, 0),
         ENTMAXKV_ERR_INVALID);
  EXPECT(entmaxkv_append_kv(&s, &a, d, mis, d, ci, ci, cd, nullptr, cf, cf, e, d, d, 0, 0),
         ENTMAXKV_ERR_INVALID);
  a.rot_dim = 0x7fffffff;
  EXPECT(entmaxkv_append_kv(&s, &a, d, d, d, ci, ci, cd, nullptr, cf, cf, e, d, d, 0, 0),
         ENTMAXKV_ERR_INVALID);
  a.rot_dim = 40;
  EXPECT(entmaxkv_append_kv(&s, &a, d, d, d, ci, ci, cd, nullptr, cf, cf, e, d, d, 0, 0),
         ENTMAXKV_ERR_UNSUPPORTED);
  a.rot_dim = 32;
  a.axes = 0x7fffffff;
  EXPECT(entmaxkv_append_kv(&s, &a, d, d, d, ci, ci, cd, ci, cf, cf, e, d, d, 0, 0),
         ENTMAXKV_ERR_INVALID);
  if (failures) return 1;
  printf("tokens driver ok\n");
  return 0;
}
