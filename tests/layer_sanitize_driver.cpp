// Host-side driver for the sanitizer build of the calls between a served layer's
// products: sizes at and past the limits and pointers at both ends of the address
// space; every call is refused before a launch, or has no tokens.  No GPU is needed
// or used.
#include <cstdint>
#include <cstdio>
#include <limits>

#include "gptq.h"

static int g_fail = 0;

#define REFUSED(call)                                                                            \
  do {                                                                                           \
    const gptq_status st = (call);                                                               \
    if (st != GPTQ_ERR_INVALID_ARG && st != GPTQ_ERR_WORKSPACE && !(st == GPTQ_OK && m == 0)) {  \
      std::fprintf(stderr, "FAILED line %d: %d\n", __LINE__, (int)st);                           \
      ++g_fail;                                                                                  \
    }                                                                                            \
  } while (0)

int main() {
  void* f = reinterpret_cast<void*>(uintptr_t{1} << 20);  // never dereferenced
  void* top = reinterpret_cast<void*>(~uintptr_t{0} - 15);
  float* ff = static_cast<float*>(f);
  int32_t* fi = static_cast<int32_t*>(f);
  int8_t* fc = static_cast<int8_t*>(f);
  const int64_t big = std::numeric_limits<int64_t>::max(), least = std::numeric_limits<int64_t>::min();
  const int64_t sizes[] = {least, -1, 0, 1, 16, 4096, 1 << 20, int64_t{1} << 30, (int64_t{1} << 30) + 1,
                           int64_t{1} << 31, (int64_t{1} << 31) + 1, int64_t{1} << 60, big};
  const gptq_integer_layer layer{fc, nullptr, fi, ff};  // without scales: refused at the latest
  size_t all = 0;
  for (int64_t m : sizes)
    for (int64_t a : sizes)
      for (int64_t b : sizes)
        for (int64_t c : {int64_t{1}, int64_t{64}, int64_t{1} << 31, big})
          for (int t : {-1, 0, 1, 2, 3}) {
            all += gptq_integer_gated_workspace_size(m, t, a, b);
            for (void* y : {f, top}) {
              REFUSED(gptq_integer_linear(f, t, ff, fi, m, a, c, &layer, b, GPTQ_ACT_SILU, y, t, c, y, 1, f, 1, nullptr));
              REFUSED(gptq_integer_linear(f, t, ff, fi, m, a, c, &layer, b, GPTQ_ACT_SILU, top, t, c, y, 1, f, 1, nullptr));
              REFUSED(gptq_integer_gated(f, t, ff, fi, m, a, c, &layer, &layer, b, GPTQ_ACT_SILU, y, t, f, 1, nullptr));
              REFUSED(gptq_norm_tokens(f, t, m, a, c, top, t, b, f, t, 1e-6f, y, c, nullptr, t, nullptr, ff, fi, nullptr));
              REFUSED(gptq_norm_tokens(f, t, m, a, c, y, t, c, f, t, 1e-6f, f, b, y, t, fc, ff, fi, nullptr));
            }
          }
  std::printf("%s (%zu)\n", g_fail ? "failures" : "all checks passed", all);
  return g_fail != 0;
}
