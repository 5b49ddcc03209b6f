// Host-only exercise of the validation and planning code of the softmax decode
// and eviction calls, built with AddressSanitizer and
// UndefinedBehaviorSanitizer (tests/test_host_sanitizers_softmax.py). Every
// call fails validation or only plans a workspace: no HIP call is reached.
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
  void* mis = reinterpret_cast<void*>((uintptr_t(1) << 20) + 8);
  const int32_t* ci = static_cast<const int32_t*>(d);
  int32_t* oi = static_cast<int32_t*>(d) + 64;
  const float* cf = static_cast<const float*>(d);
  float* of = static_cast<float*>(d);
  const size_t big = size_t(1) << 60;

  // workspace plans over the supported set, up to the largest sizes
  const int Ds[] = {64, 128}, pss[] = {16, 32, 64}, Gs[] = {1, 2, 4, 8};
  const int mps[] = {1, 7, 4096, 262144}, ns[] = {1, 2, 33, 4096, 1 << 24};
  const int Ws[] = {1, 1000, 1 << 25, 0x7fffffff}, Ss[] = {0, 4, 0x7fffffff};
  for (int D : Ds)
    for (int ps : pss)
      for (int G : Gs)
        for (int mp : mps)
          for (int dt = 0; dt < 2; ++dt)
            for (int B : {1, 16, 300, (1 << 24) / 64}) {
              const int Hkv = 8;
              if ((long long)B * Hkv * G > (1LL << 24)) continue;
              entmaxkv_shape s = {B, Hkv * G, Hkv, D, ps, mp, 0x7fffffff / ps, dt};
              size_t n = 0;
              for (int q : ns)
                for (int W : Ws)
                  for (int S : Ss) {
                    const int rc = entmaxkv_softmax_window_ws(&s, q, W, S, &n);
                    const bool fits = (long long)B * Hkv * G * q <= (1LL << 24);
                    if (rc != (fits ? ENTMAXKV_OK : ENTMAXKV_ERR_UNSUPPORTED)) ++failures;
                  }
              for (int p : {1, mp / 2 + 1, mp}) EXPECT(entmaxkv_softmax_prefix_ws(&s, p, &n), 0);
              EXPECT(entmaxkv_softmax_prefix_ws(&s, mp + 1, &n), ENTMAXKV_ERR_INVALID);
            }

  entmaxkv_shape s = {4, 32, 8, 128, 32, 4096, 16384, ENTMAXKV_BF16};
  entmaxkv_shape f = {4, 32, 8, 128, 32, 4096, 16384, ENTMAXKV_F32};
  size_t n = 0;
  EXPECT(entmaxkv_softmax_window_ws(nullptr, 1, 8, 0, &n), ENTMAXKV_ERR_INVALID);
  EXPECT(entmaxkv_softmax_window_ws(&s, 1, 8, 0, nullptr), ENTMAXKV_ERR_INVALID);
  for (int bad : {0, -1, -0x7fffffff - 1}) {
    EXPECT(entmaxkv_softmax_window(&s, d, 1, bad, d, d, ci, ci, 8, 0, d, of, d, big, 0, 0),
           ENTMAXKV_ERR_INVALID);
    EXPECT(entmaxkv_softmax_window(&s, d, 1, 1, d, d, ci, ci, bad, 0, d, of, d, big, 0, 0),
           ENTMAXKV_ERR_INVALID);
    EXPECT(entmaxkv_softmax_prefix(&s, d, 1, d, d, ci, bad, ci, ci, d, of, d, big, 0, 0),
           ENTMAXKV_ERR_INVALID);
    EXPECT(entmaxkv_evict(&s, d, d, ci, ci, cf, bad, 0, 0, oi, oi, oi, nullptr, 0, 0),
           ENTMAXKV_ERR_INVALID);
  }
  EXPECT(entmaxkv_softmax_window(&s, d, 1, 1, d, d, ci, ci, 8, -1, d, of, d, big, 0, 0),
         ENTMAXKV_ERR_INVALID);
  EXPECT(entmaxkv_softmax_window(&f, d, 1, 1, d, d, ci, ci, 8, 0, d, of, d, big, 0, 0),
         ENTMAXKV_ERR_UNSUPPORTED);
  EXPECT(entmaxkv_softmax_window(&s, mis, 1, 1, d, d, ci, ci, 8, 0, d, of, d, big, 0, 0),
         ENTMAXKV_ERR_INVALID);
  EXPECT(entmaxkv_softmax_window(&s, d, 1, 1, d, d, ci, ci, 4096, 0, d, of, nullptr, big, 0, 0),
         ENTMAXKV_ERR_WORKSPACE);
  EXPECT(entmaxkv_softmax_prefix(&s, d, 0, d, d, nullptr, 8, ci, ci, d, of, d, big, 0, 0),
         ENTMAXKV_ERR_INVALID);
  EXPECT(entmaxkv_accumulate_weights(&s, d, 0, d, ci, ci, 0.5f, cf, 8, 0, 1.0f, cf, of, 0, 0),
         ENTMAXKV_ERR_INVALID);
  EXPECT(entmaxkv_accumulate_weights(&s, d, 0, d, ci, ci, 1.5f, cf, 8, 0, NAN, cf, of, 0, 0),
         ENTMAXKV_ERR_INVALID);
  EXPECT(entmaxkv_evict(&s, d, d, ci, ci, cf, 0x7fffffff, 0, 0, oi, oi, oi, nullptr, 0, 0),
         ENTMAXKV_ERR_UNSUPPORTED);
  EXPECT(entmaxkv_evict(&s, d, d, ci, ci, cf, 8, 0x7fffffff, 0x7fffffff, oi, oi, oi, nullptr, 0, 0),
         ENTMAXKV_ERR_INVALID);
  EXPECT(entmaxkv_evict(&s, d, d, ci, ci, cf, 8, 0, 0, oi, oi, oi, of, 0, 0),
         ENTMAXKV_ERR_INVALID);  // new_weights is weights
  if (failures) return 1;
  printf("softmax driver ok\n");
  return 0;
}
